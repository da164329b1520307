"""GPU parity of the draft verification (kda_verify_drafts) with the fp64
oracle (oracle/ssm.py): whole numbers, so equality.  Products and sums are
float64 on both sides; the inputs hold no threshold within 1e-12 of a border
except where a test puts exact ones there."""
import numpy as np
import pytest

from oracle import ssm as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only container
    pytest.skip("no GPU", allow_module_level=True)

import gated_delta_rule_amd as kda  # noqa: E402


def dev(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def run(p, drafts, u, un, qd=None, nd=None, dtype=torch.float32):
    r = kda.verify_drafts(dev(p, dtype), dev(drafts, torch.int32), dev(u, torch.float32), dev(un, torch.float32),
                          dev(qd, dtype), dev(nd, torch.int32))
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in r]


def same(p, drafts, u, un, qd=None, nd=None, dtype=torch.float32):
    na, tok = run(p, drafts, u, un, qd, nd, dtype)
    for b in range(len(na)):
        n, t = O.verify(p[b], drafts[b], u[b], un[b], None if qd is None else qd[b], None if nd is None else nd[b])
        assert na[b] == n and list(tok[b]) == list(t), b
    return na


def dist(r, shape, dtype, sharp=2.0):
    z = sharp * r.standard_normal(shape)
    e = np.exp(z - z.max(-1, keepdims=True))
    p = np.float32(e / e.sum(-1, keepdims=True))
    return torch.from_numpy(p).to(dtype).float().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (3, 4, 2), (5, 3, 63), (4, 8, 4095), (4, 2, 4096), (3, 5, 4097),
                                   (2, 64, 300), (9, 0, 1000), (2, 3, 152001)])
@pytest.mark.parametrize("sampled", [True, False])
def test_parity(B, K, V, dtype, sampled):
    r = np.random.default_rng(B * 1000 + V)
    p = dist(r, (B, K + 1, V), dtype)
    qd = dist(r, (B, K, V), dtype) if sampled and K else None
    if qd is not None:
        qd[0] = p[0, :K]                       # identical: everything stands
    drafts = r.integers(0, V, (B, K)).astype(np.int32)
    if K:
        drafts[:, 0] = p[:, 0].argmax(-1)
    u, un = np.float32(r.random((B, K)) * (0.3 if sampled else 1)), np.float32(r.random(B))
    nd = r.integers(-1, K + 2, B).astype(np.int32)
    na = same(p, drafts, u, un, qd, None, dtype)
    same(p, drafts, u, un, qd, nd, dtype)
    if qd is not None:
        assert na[0] == K


def test_borders_are_exact():
    """Powers of two: every product and sum is exact, so a threshold that
    meets a border is decided by < and > alone."""
    V = 8192
    p = np.full((4, 2, V), 2.0 ** -13, np.float32)
    qd = np.zeros((4, 1, V), np.float32)
    qd[:, 0, 5] = 1.0
    drafts = np.full((4, 1), 5, np.int32)
    # u q < p fails at equality
    u = np.array([[2.0 ** -13], [np.nextafter(np.float32(2.0 ** -13), np.float32(0))], [0.0], [0.5]], np.float32)
    un = np.array([0.0, 0.5, 4096 / 8192, 0.0], np.float32)
    na = same(p, drafts, u, un, qd)
    assert list(na) == [0, 1, 1, 0]
    _, tok = run(p, drafts, u, un, qd)
    # r leaves out entry 5 in requests 0 and 3; a running sum has to pass u_next * total
    assert tok[0, 0] == 0 and tok[1, 1] == 4096 and tok[2, 1] == 4096 and tok[3, 0] == 0


def test_rows_without_mass_and_odd_values():
    V, nan, inf = 5000, float("nan"), float("inf")
    p = np.zeros((6, 2, V), np.float32)
    p[1, 0] = nan
    p[2, 0, 4500], p[2, 0, 17] = 0.25, nan              # NaN and negative entries count as zero
    p[2, 0, 3] = -1.0
    p[3, 0, 100] = 0.5                                   # q covers p: p takes r's place
    p[4, 0, 4999] = 1e-30
    p[5, 1, 42] = inf
    p[5, 0, 1] = 1.0
    qd = np.zeros((6, 1, V), np.float32)
    qd[3, 0, 100], qd[3, 0, 7] = 0.6, 0.4
    qd[2, 0, 3], qd[5, 0, 1] = 1.0, 1.0
    drafts = np.array([[0], [0], [3], [7], [1], [1]], np.int32)
    u, un = np.full((6, 1), 0.5, np.float32), np.array([0.5, 0.5, 0.999, 0.9, 0.0, 0.5], np.float32)
    na, tok = run(p, drafts, u, un, qd)
    assert list(na) == [0, 0, 0, 0, 0, 1]
    assert list(tok[:5, 0]) == [0, 0, 4500, 100, 4999] and list(tok[5]) == [1, 42]


def test_drafts_that_are_no_tokens():
    r = np.random.default_rng(3)
    p = dist(r, (3, 3, 50), torch.float32)
    drafts = np.array([[-1, 2], [50, 2], [2 ** 31 - 1, 2]], np.int32)
    u, un = np.zeros((3, 2), np.float32), np.float32(r.random(3))
    assert list(same(p, drafts, u, un)) == [0, 0, 0]
    assert list(same(p, drafts, u, un, dist(r, (3, 2, 50), torch.float32))) == [0, 0, 0]


def test_u_of_one_or_more_picks_the_last_token_with_mass():
    p = np.zeros((2, 1, 9000), np.float32)
    p[:, 0, [3, 4100, 8000]] = 0.25
    un = np.array([1.0, 2.0], np.float32)
    _, tok = run(p, np.zeros((2, 0), np.int32), np.zeros((2, 0), np.float32), un)
    assert list(tok[:, 0]) == [8000, 8000]


def test_distribution_of_many_requests():
    """Drafts drawn from q and verified: the first token follows p.  With
    65536 requests a frequency is off by at most 5 standard deviations,
    5 sqrt(p / 65536)."""
    B, V = 65536, 16
    r = np.random.default_rng(8)
    p1, q1 = dist(r, (2, V), torch.float32, 1.0), dist(r, (1, V), torch.float32, 1.0)
    drafts = r.choice(V, (B, 1), p=q1[0].astype(np.float64) / q1[0].astype(np.float64).sum()).astype(np.int32)
    na, tok = run(np.broadcast_to(p1, (B, 2, V)), drafts, np.float32(r.random((B, 1))), np.float32(r.random(B)),
                  np.broadcast_to(q1, (B, 1, V)))
    f = np.bincount(tok[:, 0], minlength=V) / B
    assert (np.abs(f - p1[0]) <= 5 * np.sqrt(p1[0] / B)).all()
    assert abs(na.mean() - np.minimum(p1[0], q1[0]).sum()) <= 5 * 0.5 / np.sqrt(B)


def test_captured_graph_replays():
    r = np.random.default_rng(9)
    p, qd = dev(dist(r, (4, 4, 9001), torch.float32), torch.float32), dev(dist(r, (4, 3, 9001), torch.float32), torch.float32)
    drafts = dev(r.integers(0, 9001, (4, 3)), torch.int32)
    u, un = torch.rand(4, 3, device="cuda") * 0.2, torch.rand(4, device="cuda")
    kda.verify_drafts(p, drafts, u, un, qd)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kda.verify_drafts(p, drafts, u, un, qd)
    for _ in range(3):
        un.uniform_()
        u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = kda.verify_drafts(p, drafts, u, un, qd)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    p = torch.full((2, 3, 8), 0.125, device="cuda")
    d, u, un = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, device="cuda"), torch.zeros(2, device="cuda")
    for bad in ((p.half(), d, u, un), (p, d.long(), u, un), (p, d, u[:1], un), (p, d, u, u), (p, d, u, un, p),
                (p.transpose(0, 1), d, u, un), (p, d, u, un, None, un)):
        with pytest.raises(kda.KDAError):
            kda.verify_drafts(*bad)
