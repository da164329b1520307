"""GPU tests of the state space calls at the edges of what their headers allow.
Tolerances as in test_gpu_ssm.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU-only container
    pytest.skip("no GPU", allow_module_level=True)

import gated_delta_rule_amd as kda  # noqa: E402
from test_gpu_ssm import check_bwd, run_bwd, scan_case  # noqa: E402

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
