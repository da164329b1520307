"""Pins of the oracle of softmax attention and of its pages (oracle/attn.py):
exact special cases, differences, and the error bounds that the GPU tests use
against float32 arithmetic."""
import numpy as np
import pytest

from oracle import attn as O


def draw(T, L, H, G, D, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((T, H, D)), r.standard_normal((L, G, D)), r.standard_normal((L, G, D))


def test_equal_scores_average_the_values():
    q, k, v = draw(5, 5, 2, 1, 4)
    o, lse = O.attention(np.zeros_like(q), k, v, 1.0)
    for t in range(5):
        assert np.allclose(o[t], v[:t + 1, 0].mean(0)) and np.allclose(lse[t], np.log(t + 1))


def test_first_token_sees_itself_only():
    q, k, v = draw(3, 3, 4, 2, 8)
    o, lse = O.attention(q, k, v, 0.5)
    assert np.allclose(o[0, :2], v[0, 0]) and np.allclose(o[0, 2:], v[0, 1])
    assert np.allclose(lse[0, 3], 0.5 * q[0, 3] @ k[0, 1])


def test_rows_that_see_nothing():
    q, k, v = draw(3, 2, 1, 1, 4)
    o, lse = O.attention(q, k, v, 1.0, first=-2)      # positions -2, -1, 0
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(o[2], v[0])
    o, lse = O.attention(q, k, v, 1.0, 0, False, there=[False, False])
    assert (o == 0).all() and np.isneginf(lse).all()


def test_parts_of_a_sequence_are_the_whole():
    q, k, v = draw(9, 9, 2, 1, 4)
    o, lse = O.attention(q, k, v, 1.0)
    o2, lse2 = O.attention(q[6:], k, v, 1.0, first=6)
    assert np.allclose(o[6:], o2) and np.allclose(lse[6:], lse2)


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_are_differences(causal):
    q, k, v = draw(6, 6, 4, 2, 3)
    gy = np.random.default_rng(1).standard_normal(q.shape)
    grads = O.attention_backward(q, k, v, gy, 0.7, causal)
    h = 1e-5
    for i, x in enumerate((q, k, v)):
        for at in [(0, 0, 0), (3, 1, 2), (5, x.shape[1] - 1, 1)]:
            f = []
            for s in (h, -h):
                y = x.copy()
                y[at] += s
                args = [q, k, v]
                args[i] = y
                f.append((O.attention(*args, 0.7, 0, causal)[0] * gy).sum())
            assert abs((f[0] - f[1]) / (2 * h) - grads[i][at]) < 1e-7


@pytest.mark.parametrize("half", [0.0, 2.0 ** -8])
def test_bounds_hold_for_float32_arithmetic(half):
    """The forms that the kernels compute, in float32 (weights rounded to bf16 where half is)."""
    torch = pytest.importorskip("torch")

    def r(x):
        return torch.from_numpy(x).float().to(torch.bfloat16).float() if half else torch.from_numpy(x).float()

    T, H, D = 40, 1, 16
    q, k, v = draw(T, T, H, 1, D, 3)
    q *= 2
    gy = np.random.default_rng(4).standard_normal(q.shape)
    q, k, v, gy = (r(x) for x in (q, k, v, gy))
    n = [x.double().numpy() for x in (q, k, v, gy)]
    x = (q[:, 0] @ k[:, 0].T) * 0.3
    x = x.masked_fill(torch.triu(torch.ones(T, T, dtype=torch.bool), 1), -float("inf"))
    m = x.max(1, keepdim=True).values
    p = torch.exp(x - m)
    low = (lambda t: t.to(torch.bfloat16).float()) if half else (lambda t: t)
    total = p.sum(1, keepdim=True)
    o = (low(p) @ v[:, 0]) / total
    lse = (m + torch.log(total))[:, 0]
    ro, rl = O.attention(*n[:3], 0.3)
    eo, el = O.bounds(*n[:3], 0.3, half)
    assert (np.abs(o.double().numpy() - ro[:, 0]) <= eo[:, 0] * 1.01).all()
    assert (np.abs(lse.double().numpy() - rl[:, 0]) <= el[:, 0]).all()
    P = torch.exp(x - lse[:, None])
    delta = (gy[:, 0] * low(o)).sum(1, keepdim=True)
    dS = low(P * (gy[:, 0] @ v[:, 0].T - delta))
    grads = 0.3 * (dS @ k[:, 0]), 0.3 * (dS.T @ q[:, 0]), low(P).T @ gy[:, 0]
    refs, errs = O.attention_backward(*n, 0.3), O.backward_bounds(*n, 0.3, half)
    for g, ref, e in zip(grads, refs, errs):
        assert (np.abs(g.double().numpy() - ref[:, 0]) <= e[:, 0] * 1.01).all()


def test_pool_by_hand():
    p = O.Pool([[-1] * 3 for _ in range(3)], [0, 0, 0], [0] * 5, 16, "abcde")
    assert p.resize([17, 1, 0]) == [1, 1, 1] and p.table == [[0, 1, -1], [2, -1, -1], [-1] * 3]
    assert p.fork([0, 0, 9], [2, 2, 1]) == [1, 0, 0]
    assert p.table[2] == [0, 3, -1] and p.refs == [2, 1, 1, 1, 0] and p.data[3] == "b"
    assert p.resize([0, 40, 17]) == [1, 1, 1] and p.table[1] == [2, 1, 4] and p.refs == [1, 1, 1, 1, 1]
    assert p.resize([0, 0, 17]) == [1, 1, 1]
    assert p.compact() == ([[-1] * 3, [-1] * 3, [0, 1, -1]], [1, 1, 0, 0, 0], 2) and p.data[1] == "b"


def test_pairs_that_copy_nothing_need_no_page():
    table = [[0, -1], [1, -1], [2, 3], [-1, -1], [-1, -1], [4, 5]]
    p = O.Pool(table, [10, 16, 32, 0, 0, 20], [1] * 6, 16, "abcdef")
    assert p.fork([0, 1, 0, 5, 3], [3, 4, 5, 5, 2]) == [0, 1, 0, 0, 1]
    assert p.table == [[0, -1], [1, -1], [-1, -1], [-1, -1], [1, -1], [4, 5]]
    assert p.lengths == [10, 16, 0, 0, 16, 20] and p.refs == [1, 2, 0, 0, 1, 1] and p.data == list("abcdef")
    assert p.fork([0, 5, 0, 5, 1], [2, 3, 4, 5, 1]) == [1, 1, 0, 1, 1]
    assert p.table == [[0, -1], [1, -1], [2, -1], [4, 3], [1, -1], [4, 5]]
    assert p.lengths == [10, 16, 10, 20, 16, 20] and p.refs == [1, 2, 1, 1, 2, 1] and p.data == list("abafef")
