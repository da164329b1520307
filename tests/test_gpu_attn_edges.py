"""Softmax attention and its paged cache at the sizes and in the uses where they
could go wrong: long requests and many of them (cut into pieces), offsets past
32 bits, captured graphs, other streams, a serving run of all calls together.

Expected values are plain float64 on the GPU; tolerances are the bounds of
oracle/attn.py (see tests/test_gpu_attn.py), in the same float64.
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
U = 2.0 ** -24


def exact(q, K, V, first, scale, dtype, causal=True):
    """o, lse of one sequence's queries [T, H, D] over keys [L, G, D] in float64,
    and the largest errors of float32 arithmetic with weights rounded once."""
    T, H, D = q.shape
    L, G = K.shape[:2]
    half = 2.0 ** -8 if dtype == BF16 else 0.0
    out = [torch.zeros(T, H, D, dtype=torch.float64, device="cuda") for _ in range(2)]
    out += [torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2)]
    late = torch.arange(L, device="cuda")[None] > first + torch.arange(T, device="cuda")[:, None]
    for h in range(H):
        k, v = K[:, h // (H // G)].double(), V[:, h // (H // G)].double()
        qh = q[:, h].double()
        x = (qh @ k.T.contiguous()) * scale
        mag = abs(scale) * (qh.abs() @ k.abs().T.contiguous())
        if causal:
            x, mag = x.masked_fill(late, -float("inf")), mag.masked_fill(late, 0.0)
        lse = torch.logsumexp(x, 1)
        P = torch.exp(x - lse[:, None]).masked_fill(torch.isneginf(lse)[:, None], 0.0)   # (rows that see nothing)
        s = mag.amax(1) * (D + 8) * U
        out[0][:, h], out[2][:, h] = P @ v, lse
        out[1][:, h] = (half + 2 * s + (L + 32) * U)[:, None] * (P @ v.abs())
        out[3][:, h] = s + (lse.masked_fill(torch.isneginf(lse), 0.0).abs() + L + 32) * U
    return out


def check(name, got, ref, err, dtype):
    none = torch.isneginf(ref)
    assert torch.equal(torch.isneginf(got), none), name
    got, ref = got.double().masked_fill(none, 0.0), ref.masked_fill(none, 0.0)
    tol = err * 1.01 + (2.0 ** -8 if dtype == BF16 else U) * ref.abs() * 1.01 + 1e-30
    worst = float(((got - ref).abs() / tol).max())
    assert worst <= 1.0, f"{name}: {worst:.3g} of the tolerance"
    return worst


class Cache:
    """Requests with random keys and values in shuffled pages."""

    def __init__(self, held, G, D, page, dtype, seed=0, room=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        count = [-(-(h + room) // page) for h in held]
        n = sum(count) + 2
        self.kp = torch.randn(n, G, page, D, generator=g, device="cuda").to(dtype)
        self.vp = torch.randn(n, G, page, D, generator=g, device="cuda").to(dtype)
        order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(held), max(count + [1])), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(count):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.lengths = torch.tensor(held, dtype=torch.int32, device="cuda")
        self.held, self.page = held, page

    def keys(self, b):
        rows = self.table[b, :-(-self.held[b] // self.page)].long()
        return [t[rows].transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])[:self.held[b]] for t in (self.kp, self.vp)]


def run_paged(held, new, H, G, D, page, dtype, seed=0, look=None, scale=None):
    c = Cache(held, G, D, page, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    T = sum(new)
    q = (1.5 * torch.randn(T, H, D, generator=g, device="cuda")).to(dtype)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    equal = len(set(new)) == 1
    if equal:
        o, lse = kda.attn_paged_fwd(q.view(len(new), new[0], H, D), c.kp, c.vp, c.table, c.lengths, scale=scale)
        o, lse = o.view(T, H, D), lse.view(T, H)
    else:
        o, lse = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths, cu, scale=scale)
    w, at = 0.0, 0
    for b, t in enumerate(new):
        if t and (look is None or b in look):
            K, V = c.keys(b)
            ref, eo, lref, el = exact(q[at:at + t], K, V, held[b] - t, D ** -0.5 if scale is None else scale, dtype)
            w = max(w, check(f"o {b}", o[at:at + t], ref, eo, dtype), check(f"lse {b}", lse[at:at + t], lref, el, F32))
        at += t
    say(f"[paged] {len(held)} requests up to {max(held)}, {T} rows, {H}/{G} x {D} {dtype}: {w:.2g} of the tolerance")


STEPS = [([70000], [1], 8, 2, 128, 64), ([33000, 1, 40000, 500], [3] * 4, 15, 3, 64, 16), ([9000, 5000], [16, 16], 16, 4, 128, 256),
         ([20001], [21], 6, 2, 64, 32), ([3000, 77], [64, 64], 2, 2, 128, 16)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", STEPS)
def test_few_rows_over_long_requests(case, dtype):
    run_paged(*case, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_requests_than_threads(dtype):
    r = np.random.default_rng(0)
    held = [int(x) for x in r.integers(1, 300, 600)]
    held[7] = 9000
    run_paged(held, [1] * 600, 4, 2, 64, 16, dtype, look={0, 7, 8, 255, 256, 257, 300, 511, 512, 598, 599})


BLOCKS = [([30000, 4000], [150, 333], 8, 2, 128, 16), ([5000], [700], 4, 4, 64, 64), ([2500, 2500, 2500], [100, 100, 100], 12, 3, 128, 32),
          ([20000], [65], 1, 1, 128, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", BLOCKS)
def test_chunks_over_long_requests(case, dtype):
    run_paged(*case, dtype)


MIXED = [([5000] + [700] * 20 + [90, 2000, 31], [1] * 21 + [0, 257, 5], 8, 2, 128, 64), ([300] * 70, [1] * 69 + [2], 4, 4, 64, 16),
         ([9000, 9000, 40], [1, 130, 33], 32, 2, 64, 32)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", MIXED)
def test_single_tokens_beside_chunks(case, dtype):
    run_paged(*case, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,G,lens", [(200, 1, [37, 5]), (130, 2, [3, 0, 21])])
def test_many_heads_to_a_group(H, G, lens, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    T, D = sum(lens), 64
    q, k, v, go = (torch.randn(T, n, D, generator=g, device="cuda").to(dtype) for n in (H, G, G, H))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o, lse = kda.attn_fwd(q, k, v, cu)
    grads = kda.attn_bwd(q, k, v, o, lse, go, cu)
    at = 0
    for t in lens:
        if t:
            s = slice(at, at + t)
            ref, eo, lref, el = exact(q[s], k[s], v[s], 0, D ** -0.5, dtype)
            check("o", o[s], ref, eo, dtype)
            check("lse", lse[s], lref, el, F32)
            n = [x[s].double().cpu().numpy() for x in (q, k, v, go)]
            refs, errs = O.attention_backward(*n, D ** -0.5), O.backward_bounds(*n, D ** -0.5, 2.0 ** -8 if dtype == BF16 else 0.0)
            for x, r, e in zip(grads, refs, errs):
                check("gradient", x[s], torch.from_numpy(r).cuda(), torch.from_numpy(e).cuda(), dtype)
        at += t
    run_paged([400, 70], [3, 70], H, G, D, 16, dtype)


def test_many_blocks_are_not_cut():
    run_paged([1200] * 9, [900] * 9, 16, 8, 64, 16, BF16, look={0, 4, 8})


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
@pytest.mark.parametrize("new", [[2, 2], [90, 90]])
def test_scales(new, scale, dtype):
    run_paged([300, 120], new, 4, 2, 64, 16, dtype, scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_scales_of_prompts(scale, dtype):
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, go = (torch.randn(1, 150, n, 64, generator=g, device="cuda").to(dtype) for n in (4, 2, 2, 4))
    o, lse = kda.attn_fwd(q, k, v, scale=scale)
    ref, eo, lref, el = exact(q[0], k[0], v[0], 0, scale, dtype)
    check("o", o[0], ref, eo, dtype)
    check("lse", lse[0], lref, el, F32)
    n = [t[0].double().cpu().numpy() for t in (q, k, v, go)]
    refs, errs = O.attention_backward(*n, scale), O.backward_bounds(*n, scale, 2.0 ** -8 if dtype == BF16 else 0.0)
    for x, r, e in zip(kda.attn_bwd(q, k, v, o, lse, go, scale=scale), refs, errs):
        check("gradient", x[0], torch.from_numpy(r).cuda(), torch.from_numpy(e).cuda(), dtype)


@pytest.mark.parametrize("T", [8, 50, 150])
def test_grad_k_does_not_depend_on_the_rounding_of_o(T):
    # values of 128 and a little: bf16 holds o to 0.5 only, and delta = grad_o . o to about 0.15 |grad_o|
    g = torch.Generator(device="cuda").manual_seed(T)
    D = 64
    q, k, go = (torch.randn(1, T, 1, D, generator=g, device="cuda").to(BF16) for _ in range(3))
    v = (128 + torch.randint(0, 4, (1, T, 1, D), generator=g, device="cuda")).to(BF16)
    o, lse = kda.attn_fwd(q, k, v)
    gk = kda.attn_bwd(q, k, v, o, lse, go)[1][0, :, 0].double()
    q, k, v, go = (t[0, :, 0].double() for t in (q, k, v, go))
    late = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
    x = (q @ k.T.contiguous() * D ** -0.5).masked_fill(late, -float("inf"))
    P, dP = torch.softmax(x, 1), go @ v.T.contiguous()
    dS = P * (dP - (P * dP).sum(1, keepdim=True))
    # P: errors of scores and lse in float32; dP and the sum of dS: of products of 64 float32 terms and sums over the row
    score = D ** -0.5 * (q.abs() @ k.abs().T.contiguous()).amax(1) * (D + 8) * U
    part = (go.abs() @ v.abs().T.contiguous()).amax(1) * (2 * D + T + 16) * U
    err = dS.abs() * (2.0 ** -8 + (4 * score + (T + 40) * U)[:, None]) + 2 * P * part[:, None]
    ref = D ** -0.5 * (dS.T.contiguous() @ q)
    check("grad_k", gk, ref, D ** -0.5 * (err.T.contiguous() @ q.abs()), BF16)


@pytest.mark.parametrize("dtype,n,T,H,G,D", [(BF16, 1, 5000, 4, 1, 128), (BF16, 3, 1111, 8, 8, 64), (F32, 1, 2100, 4, 2, 128)])
def test_long_prompts(dtype, n, T, H, G, D):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, go = (torch.randn(n, T, m, D, generator=g, device="cuda").to(dtype) for m in (H, G, G, H))
    o, lse = kda.attn_fwd(q, k, v)
    grads = kda.attn_bwd(q, k, v, o, lse, go)
    half, scale = 2.0 ** -8 if dtype == BF16 else 0.0, D ** -0.5
    late = torch.triu(torch.ones(T, T, dtype=torch.bool, device="cuda"), 1)
    for b in range(n):
        ref, eo, lref, el = exact(q[b], k[b], v[b], 0, scale, dtype)
        check("o", o[b], ref, eo, dtype)
        check("lse", lse[b], lref, el, F32)
        gq, gk, gv = (torch.zeros(t.shape[1:], dtype=torch.float64, device="cuda") for t in (q, k, v))
        eq, ek, ev = (torch.zeros_like(t) for t in (gq, gk, gv))
        for h in range(H):   # as oracle/attn.py: attention_backward and backward_bounds
            i = h // (H // G)
            Q, K, V, Y = q[b, :, h].double(), k[b, :, i].double(), v[b, :, i].double(), go[b, :, h].double()
            P = torch.exp(((Q @ K.T.contiguous()) * scale).masked_fill(late, -float("inf")) - lref[:, h:h + 1])
            gP, O = Y @ V.T.contiguous(), P @ V
            delta, dmag = (Y * O).sum(1, keepdim=True), (Y.abs() * O.abs()).sum(1, keepdim=True)
            gS = P * (gP - delta)
            gq[:, h] = scale * gS @ K
            gk[:, i] += scale * gS.T.contiguous() @ Q
            gv[:, i] += P.T.contiguous() @ Y
            s = (scale * (Q.abs() @ K.abs().T.contiguous())).masked_fill(late, 0.0).amax(1) * (D + 8) * U
            rel = (2 * s + s + (P.amax(1).log().abs() + T + 64) * U + 64 * U)[:, None]
            n_sum = (T * (H // G) + 32) * U
            eS = P * (half * ((gP - delta).abs() + dmag) * 1.02 + (rel + (D + 8) * U) * (Y.abs() @ V.abs().T.contiguous() + dmag))
            eS = eS + n_sum * P * ((gP - delta).abs() + half * dmag)
            eq[:, h] = scale * eS @ K.abs()
            ek[:, i] += scale * eS.T.contiguous() @ Q.abs()
            ev[:, i] += (P * (half + rel + n_sum)).T.contiguous() @ Y.abs()
        w = [check(name, x[b], r, e, dtype) for name, x, r, e in zip(("gq", "gk", "gv"), grads, (gq, gk, gv), (eq, ek, ev))]
    say(f"[prompt] {n} x {T}, {H}/{G} x {D} {dtype}: gradients at {max(w):.2g} of the tolerance")


def test_offsets_past_32_bits():
    # pages of a pool whose elements are counted past 2^32
    G, D, page = 2, 64, 16
    stride = 1 << 27
    pool = torch.empty(40, stride, dtype=BF16, device="cuda")       # 10.7 GB
    size = G * page * D
    kp, vp = (pool[:, i * size:(i + 1) * size].unflatten(1, (G, page, D)) for i in range(2))
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (kp, vp):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    table = torch.tensor([[39, 0, 38, 33], [34, 37, 36, 35]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([64, 50], dtype=torch.int32, device="cuda")
    small = [t[table.long().flatten()].contiguous() for t in (kp, vp)]
    near = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    for T in (1, 3, 40):
        q = torch.randn(2, T, 4, D, generator=g, device="cuda").to(BF16)
        new = [torch.randn(2, T, G, D, generator=g, device="cuda").to(BF16) for _ in range(2)]
        kda.kv_append(*new, kp, vp, table, lengths)
        kda.kv_append(*new, *small, near, lengths)
        assert torch.equal(kp[table.long().flatten()], small[0]) and torch.equal(vp[table.long().flatten()], small[1])
        a, b = kda.attn_paged_fwd(q, kp, vp, table, lengths), kda.attn_paged_fwd(q, *small, near, lengths)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a branch of the first request: its open page is copied from far to far
    table3, lengths3 = torch.full((3, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    table3[:2], lengths3[:2] = table, lengths
    refs = torch.ones(40, dtype=torch.int32, device="cuda")
    refs[32] = 0
    ok = kda.kv_fork(table3, lengths3, refs, torch.tensor([1], dtype=torch.int32, device="cuda"),
                     torch.tensor([2], dtype=torch.int32, device="cuda"), (kp, vp), page)
    assert ok.tolist() == [1] and table3[2].tolist() == [34, 37, 36, 32]
    assert torch.equal(kp[32], kp[35]) and torch.equal(vp[32], vp[35])


class Server:
    """A layer of attention over a pool, its state on the device."""

    def __init__(self, slots, n_pages, most, G, D, page, dtype, device="cuda"):
        self.pool = torch.full((n_pages, 2, G, page, D), float("nan"), dtype=dtype, device=device)
        self.kp, self.vp = self.pool[:, 0], self.pool[:, 1]
        self.table = torch.full((slots, most), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(slots, dtype=torch.int32, device=device)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=device)
        self.page = page

    def step(self, q, k, v, want):
        ok = kda.kv_resize(self.table, self.lengths, self.refs, want, self.page)
        kda.kv_append(k, v, self.kp, self.vp, self.table, self.lengths)
        o, lse = kda.attn_paged_fwd(q, self.kp, self.vp, self.table, self.lengths)
        return ok, o, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_serving_run(dtype):
    """Prompts in chunks, branches, drafts with their verification and rollback,
    compaction: the tokens that stay see what one prompt call says."""
    G, D, H, page, slots = 2, 64, 6, 16, 4
    s = Server(slots, 40, 8, G, D, page, dtype)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rows(T):
        return [torch.randn(slots, T, n, D, generator=g, device="cuda").to(dtype) for n in (H, G, G)]

    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    seen = [[] for _ in range(slots)]   # of each slot: rows of q, k, v and the outputs they got

    def step(T, kept):
        """T new tokens in every slot, of which kept[b] stay."""
        q, k, v = rows(T)
        ok, o, lse = s.step(q, k, v, s.lengths + T)
        assert ok.tolist() == [1] * slots
        for b in range(slots):
            seen[b] += [(q[b, t], k[b, t], v[b, t], o[b, t], lse[b, t]) for t in range(kept[b])]
        if min(kept) < T:
            kda.kv_resize(s.table, s.lengths, s.refs, ints([len(x) for x in seen]), page)

    step(37, [37] * slots)                                   # a chunk of a prompt
    step(1, [1] * slots)
    p = torch.softmax(torch.randn(slots, 4, 50, generator=g, device="cuda"), -1)
    drafts = torch.randint(0, 50, (slots, 3), generator=g, device="cuda").to(torch.int32)
    u = torch.rand(slots, 3, generator=g, device="cuda") * 0.05
    n_acc, _ = kda.verify_drafts(p, drafts, u, u[:, 0].contiguous())
    step(4, [1 + int(n) for n in n_acc.tolist()])            # the token before the drafts, and those that stand
    kda.kv_fork(s.table, s.lengths, s.refs, ints([0, 0, 3]), ints([1, 2, 3]), s.pool, page)
    seen = [list(seen[0]), list(seen[0]), list(seen[0]), seen[3]]
    step(5, [5, 2, 0, 4])
    kda.kv_compact(s.table, s.lengths, s.refs, s.pool, page, table_out=s.table, refs_out=s.refs)
    step(3, [3] * slots)
    for b in range(slots):
        q, k, v, o, lse = (torch.stack(x) for x in zip(*seen[b]))
        ref, eo, lref, el = exact(q, k, v, 0, D ** -0.5, dtype)
        check("o", o, ref, eo, dtype)
        check("lse", lse, lref, el, F32)
        whole, _ = kda.attn_fwd(q[None], k[None], v[None])
        check("prompt", whole[0], ref, eo, dtype)
    held = [-(-len(x) // page) for x in seen]
    assert s.lengths.tolist() == [len(x) for x in seen]
    used = [p for b in range(slots) for p in s.table[b, :held[b]].tolist()]
    assert s.refs.tolist() == [used.count(p) for p in range(40)]
    kda.kv_resize(s.table, s.lengths, s.refs, ints([0] * slots), page)
    assert int(s.refs.abs().sum()) == 0 and (s.table == -1).all()


def test_captured_serving_step():
    """A step captured into a graph, replayed with other inputs, lengths and tables
    between eager work, against the same eager steps; two graphs in turn."""
    G, D, H, page, slots, T = 2, 128, 8, 16, 3, 2
    a, b = (Server(slots, 60, 16, G, D, page, BF16) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(4)
    ins = [torch.zeros(slots, T, n, D, dtype=BF16, device="cuda") for n in (H, G, G)]
    want = torch.zeros(slots, dtype=torch.int32, device="cuda")
    src, dst = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")

    def body(s):
        out = s.step(*ins, want)
        kda.kv_fork(s.table, s.lengths, s.refs, src, dst, s.pool, page)
        kda.kv_compact(s.table, s.lengths, s.refs, s.pool, page, table_out=s.table, refs_out=s.refs)
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body(a)
    torch.cuda.current_stream().wait_stream(side)
    kda.kv_resize(a.table, a.lengths, a.refs, torch.zeros_like(want), page)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = body(a)
        graphs.append((graph, out))
    kda.kv_resize(a.table, a.lengths, a.refs, torch.zeros_like(want), page)
    a.pool.fill_(0)
    b.pool.fill_(0)
    kda.kv_resize(b.table, b.lengths, b.refs, torch.zeros_like(want), page)
    for i in range(8):
        for t in ins:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        want.copy_(torch.randint(2, 200, (slots,), generator=g, device="cuda"))
        src.fill_(i % slots)
        dst.fill_((i + 1) % slots)
        graph, out = graphs[i % 2]
        graph.replay()
        eager = body(b)
        torch.cuda.synchronize()
        for x, y in zip(out, eager):
            assert torch.equal(x.nan_to_num(3.0, 4.0, 5.0), y.nan_to_num(3.0, 4.0, 5.0)), i
        for x, y in ((a.table, b.table), (a.lengths, b.lengths), (a.refs, b.refs), (a.pool, b.pool)):
            assert torch.equal(x, y), i


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_training_step(dtype):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, go = (torch.randn(2, 200, n, 64, generator=g, device="cuda").to(dtype) for n in (8, 2, 2, 8))

    def body():
        o, lse = kda.attn_fwd(q, k, v)
        return (o, lse) + kda.attn_bwd(q, k, v, o, lse, go)

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = body()
    for i in range(4):
        for t in (q, k, v, go):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        eager = body()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, eager)), i


def test_another_stream_and_two_calls_at_once():
    g = torch.Generator(device="cuda").manual_seed(6)
    sets = []
    for n in (2, 3):
        c = Cache([900, 40, 3000][:n], 2, 128, 16, BF16, n)
        q = torch.randn(n, 2, 8, 128, generator=g, device="cuda").to(BF16)
        x = [torch.randn(1, 700, m, 64, generator=g, device="cuda").to(BF16) for m in (4, 2, 2, 4)]
        sets.append((c, q, x))

    def work(c, q, x):
        o, lse = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths)
        p, plse = kda.attn_fwd(*x[:3])
        return (o, lse, p, plse) + kda.attn_bwd(*x[:3], p, plse, x[3])

    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(work(*s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_results_repeat_bitwise():
    c = Cache([5000, 100, 2222], 4, 64, 32, BF16, 9)
    for T in (1, 7, 100):
        q = torch.randn(3, T, 8, 64, device="cuda").to(BF16)
        first = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths)
        for _ in range(3):
            again = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths)
            assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_empty_batches(dtype):
    kv = torch.empty(0, 5, 2, 64, dtype=dtype, device="cuda")
    q = torch.empty(0, 5, 4, 64, dtype=dtype, device="cuda")
    o, lse = kda.attn_fwd(q, kv, kv)
    assert o.shape == q.shape and lse.shape == (0, 5, 4)
    assert [t.shape for t in kda.attn_bwd(q, kv, kv, o, lse, q)] == [q.shape, kv.shape, kv.shape]
    q, kv = q.view(5, 0, 4, 64), kv.view(5, 0, 2, 64)
    assert kda.attn_fwd(q, kv, kv)[0].shape == q.shape
    c = Cache([3] * 5, 2, 64, 16, dtype)
    assert kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths)[0].shape == q.shape
    # packed, without sequences: nothing is a row of one
    q, kv = torch.ones(6, 4, 64, dtype=dtype, device="cuda"), torch.ones(6, 2, 64, dtype=dtype, device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = kda.attn_fwd(q, kv, kv, none)
    grads = kda.attn_bwd(q, kv, kv, o, lse, q, none)
    assert all((t == 0).all() for t in grads)
    # requests that hold nothing at all
    c.lengths.zero_()
    o, lse = kda.attn_paged_fwd(torch.ones(5, 2, 4, 64, dtype=dtype, device="cuda"), c.kp, c.vp, c.table, c.lengths)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = kda.attn_paged_fwd(torch.ones(5, 40, 4, 64, dtype=dtype, device="cuda"), c.kp, c.vp, c.table, c.lengths)
    assert (o == 0).all() and torch.isneginf(lse).all()


# held, new, H, G, D, page: steps in one piece and cut, chunks taken whole, cut and in parts
NAN_ROWS = [([40, 7], [2, 2], 4, 2, 64, 16), ([9000], [1], 8, 2, 128, 64), ([9000, 300], [4, 4], 64, 4, 64, 64), ([300, 80], [70, 70], 4, 2, 64, 16),
            ([20000], [150], 8, 2, 128, 16)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", NAN_ROWS)
def test_lse_says_nan_beside_a_nan(case, dtype):
    """A NaN in a query, or in a key that it sees, is no row that sees nothing."""
    held, new, H, G, D, page = case
    c, n, T = Cache(held, G, D, page, dtype), len(held), new[0]
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(n, T, H, D, generator=g, device="cuda").to(dtype)
    bad = torch.zeros(n, T, H, dtype=torch.bool, device="cuda")
    bad[0, T // 2, H - 1] = bad[n - 1, T - 1, 0] = True
    refs = [exact(q[b], *c.keys(b), held[b] - T, D ** -0.5, dtype) for b in range(n)]
    q[bad] = float("nan")
    o, lse = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths)
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(o).all(-1), bad)
    for b, (ref, eo, lref, el) in enumerate(refs):
        check("o", o[b][~bad[b]], ref[~bad[b]], eo[~bad[b]], dtype)
        check("lse", lse[b][~bad[b]], lref[~bad[b]], el[~bad[b]], F32)
    # one value of the first key of request 0, group 0
    c.kp[c.table[0, 0].long(), 0, 0, D - 1] = float("nan")
    o, lse = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths)
    bad[0, :, :H // G] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(o).all(-1), bad)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lse_of_a_prompt_says_nan_beside_a_nan(dtype):
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (torch.randn(2, 150, n, 64, generator=g, device="cuda").to(dtype) for n in (4, 2, 2))
    q[0, 30, 1, 5], k[1, 100, 1, 9] = float("nan"), float("nan")
    bad = torch.zeros(2, 150, 4, dtype=torch.bool, device="cuda")
    bad[0, 30, 1] = bad[1, 100:, 2:] = True
    o, lse = kda.attn_fwd(q, k, v)
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(o).all(-1), bad)
    assert not torch.isinf(lse).any()


def unseen(o, lse, q, K, V, first, dtype, at, d, what):
    """Rows before key `at` are as if it held no `what` in value d; from it on that value is `what`."""
    D = q.shape[-1]
    ref, eo, lref, el = exact(q, K, V.nan_to_num(0.0, 0.0, 0.0), first, D ** -0.5, dtype)
    H, G = q.shape[1], K.shape[1]
    bad = torch.zeros(ref.shape, dtype=torch.bool, device="cuda")
    bad[max(0, at - first):, -(H // G):, d] = True       # (the last group)
    got = o.masked_select(bad)
    assert torch.isnan(got).all() if what != what else (got == what).all()
    check("o", o.masked_fill(bad, 0.0), ref.masked_fill(bad, 0.0), eo, dtype)
    check("lse", lse, lref, el, F32)


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,at,H,G,D", [([5], 4, 2, 1, 64), ([70, 300], 250, 8, 2, 128), ([64, 129], 1, 3, 3, 64), ([600], 599, 4, 1, 64),
                                           ([300, 200, 90], 63, 4, 4, 128)])
def test_a_value_that_is_not_finite_reaches_no_earlier_row(lens, at, H, G, D, dtype, what):
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(sum(lens), n, D, generator=g, device="cuda").to(dtype) for n in (H, G, G))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    last = slice(sum(lens[:-1]), sum(lens))
    v[last][at, G - 1, 7] = what
    o, lse = kda.attn_fwd(q, k, v, cu)
    for n, s in zip(lens, cu.tolist()):
        x = slice(s, s + n)
        unseen(o[x], lse[x], q[x], k[x], v[x], 0, dtype, at if x == last else n, 7, what)


@pytest.mark.parametrize("what", [float("nan"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", [([40, 7], [3, 3], 4, 2, 64, 16), ([9000], [5], 8, 2, 128, 64), ([9000, 300], [4, 4], 64, 4, 64, 64),
                                  ([300, 80], [70, 70], 4, 2, 64, 16), ([20000], [150], 8, 2, 128, 16), ([700, 900], [200, 30], 8, 2, 128, 32)])
def test_a_new_value_that_is_not_finite_reaches_no_earlier_row(case, dtype, what):
    held, new, H, G, D, page = case
    c, n = Cache(held, G, D, page, dtype), len(held)
    g = torch.Generator(device="cuda").manual_seed(10)
    q = torch.randn(sum(new), H, D, generator=g, device="cuda").to(dtype)
    x = held[-1] - new[-1] // 2
    c.vp[c.table[n - 1, x // page].long(), G - 1, x % page, D - 1] = what
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    o, lse = kda.attn_paged_fwd(q, c.kp, c.vp, c.table, c.lengths, cu)
    for b in range(n):
        s = slice(int(cu[b]), int(cu[b + 1]))
        unseen(o[s], lse[s], q[s], *c.keys(b), held[b] - new[b], dtype, x if b == n - 1 else held[b], D - 1, what)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_padding_may_hold_anything(dtype):
    # equal lengths, of which the batch's sequences fill less: their tokens see no padding
    g = torch.Generator(device="cuda").manual_seed(11)
    lens, T, H, G, D = [200, 1, 131, 64], 200, 6, 2, 64
    q, k, v = (torch.randn(len(lens), T, n, D, generator=g, device="cuda").to(dtype) for n in (H, G, G))
    for b, n in enumerate(lens):
        for t in (q, k, v):
            t[b, n:] = float("nan")
    o, lse = kda.attn_fwd(q, k, v)
    for b, n in enumerate(lens):
        ref, eo, lref, el = exact(q[b, :n], k[b, :n], v[b, :n], 0, D ** -0.5, dtype)
        check("o", o[b, :n], ref, eo, dtype)
        check("lse", lse[b, :n], lref, el, F32)
        assert torch.isnan(o[b, n:]).all() and torch.isnan(lse[b, n:]).all()


@pytest.mark.parametrize("held,new", [
    # uneven lengths, cut into pieces: single tokens, a chunk, requests without new tokens
    ([100 + 37 * (b % 11) for b in range(150)] + [20000] + [60] * 110 + [9000, 300] + [500] * 60, [1] * 100 + [0, 1] * 25 + [150] + [1] * 170 + [0, 2]),
    # short ones, taken whole
    ([40 + b % 7 for b in range(330)], [1] * 329 + [9])])
def test_more_blocks_than_threads(held, new):
    """More than 256 blocks per group: a thread of the piece finding has several."""
    cu = np.concatenate([[0], np.cumsum(new)])
    slots = cu[:-1] * 8 // 128 + np.arange(len(new))      # first block of each request
    assert slots[-1] > 256 and (cu[-1] * 8 // 128 + len(new)) * 4 < 2048
    look = {0, 1, 99, 149, 150, 151, 200, 261, 262, len(new) - 2, len(new) - 1} | set(np.nonzero((slots >= 250) & (slots < 262))[0].tolist())
    run_paged(held, new, 32, 4, 64, 16, BF16, look=look)


@pytest.mark.parametrize("dtype,n,T,H,G,D", [(BF16, 1, 2100, 4, 2, 128), (BF16, 2, 1111, 6, 2, 64), (F32, 1, 1300, 4, 2, 128), (F32, 2, 700, 3, 3, 64)])
def test_long_sequences_that_see_all(dtype, n, T, H, G, D):
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k, v, go = (torch.randn(n, T, m, D, generator=g, device="cuda").to(dtype) for m in (H, G, G, H))
    o, lse = kda.attn_fwd(q, k, v, causal=False)
    grads = kda.attn_bwd(q, k, v, o, lse, go, causal=False)
    half, scale = 2.0 ** -8 if dtype == BF16 else 0.0, D ** -0.5
    for b in range(n):
        ref, eo, lref, el = exact(q[b], k[b], v[b], 0, scale, dtype, causal=False)
        check("o", o[b], ref, eo, dtype)
        check("lse", lse[b], lref, el, F32)
        refs = [torch.zeros(t.shape[1:], dtype=torch.float64, device="cuda") for t in (q, k, v)]
        errs = [torch.zeros_like(t) for t in refs]
        for h in range(H):   # as oracle/attn.py: attention_backward and backward_bounds
            i = h // (H // G)
            Q, K, V, Y = q[b, :, h].double(), k[b, :, i].double(), v[b, :, i].double(), go[b, :, h].double()
            P = torch.exp((Q @ K.T.contiguous()) * scale - lref[:, h:h + 1])
            gP, out = Y @ V.T.contiguous(), P @ V
            delta, dmag = (Y * out).sum(1, keepdim=True), (Y.abs() * out.abs()).sum(1, keepdim=True)
            gS = P * (gP - delta)
            refs[0][:, h] = scale * gS @ K
            refs[1][:, i] += scale * gS.T.contiguous() @ Q
            refs[2][:, i] += P.T.contiguous() @ Y
            s = (scale * (Q.abs() @ K.abs().T.contiguous())).amax(1) * (D + 8) * U
            rel = (3 * s + (P.amax(1).log().abs() + T + 128) * U)[:, None]
            n_sum = (T * (H // G) + 32) * U
            eS = P * (half * ((gP - delta).abs() + dmag) * 1.02 + (rel + (D + 8) * U) * (Y.abs() @ V.abs().T.contiguous() + dmag))
            eS = eS + n_sum * P * ((gP - delta).abs() + half * dmag)
            errs[0][:, h] = scale * eS @ K.abs()
            errs[1][:, i] += scale * eS.T.contiguous() @ Q.abs()
            errs[2][:, i] += (P * (half + rel + n_sum)).T.contiguous() @ Y.abs()
        w = [check(name, x[b], r, e, dtype) for name, x, r, e in zip(("gq", "gk", "gv"), grads, refs, errs)]
    say(f"[all] {n} x {T}, {H}/{G} x {D} {dtype}: gradients at {max(w):.2g} of the tolerance")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,G,D,share", [(400, 6, 2, 64, 0.002), (333, 4, 4, 128, 0.0005), (700, 8, 1, 128, 0.00005), (200, 3, 1, 64, 0.2)])
def test_values_that_are_not_finite_here_and_there(T, H, G, D, share, dtype):
    """Each value of a row is a NaN if a token that it sees has one there, else as if there was none: of a prompt, and of its
    last tokens over a cache."""
    g = torch.Generator(device="cuda").manual_seed(13)
    q, k, v = (torch.randn(T, n, D, generator=g, device="cuda").to(dtype) for n in (H, G, G))
    v[torch.rand(T, G, D, generator=g, device="cuda") < share] = float("nan")
    v[T - 1, 0, 1] = v[T - 30, G - 1, D - 2] = float("nan")
    ref, eo, lref, el = exact(q, k, v.nan_to_num(0.0), 0, D ** -0.5, dtype)
    had = torch.isnan(v).cumsum(0).bool().repeat_interleave(H // G, 1)
    o, lse = kda.attn_fwd(q[None], k[None], v[None])
    assert torch.equal(torch.isnan(o[0]), had)
    check("o", o[0].nan_to_num(0.0), ref.masked_fill(had, 0.0), eo, dtype)
    check("lse", lse[0], lref, el, F32)
    page = 16
    n_pages = -(-T // page)
    kp, vp = (torch.full((n_pages, G, page, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)[None]
    lengths = torch.tensor([T], dtype=torch.int32, device="cuda")
    kda.kv_append(k[None], v[None], kp, vp, table, lengths)
    for new in (2, 7, 60, T):
        o, lse = kda.attn_paged_fwd(q[None, T - new:], kp, vp, table, lengths)
        assert torch.equal(torch.isnan(o[0]), had[T - new:]), new
        check("o", o[0].nan_to_num(0.0), ref[T - new:].masked_fill(had[T - new:], 0.0), eo[T - new:], dtype)
        check("lse", lse[0], lref[T - new:], el[T - new:], F32)
