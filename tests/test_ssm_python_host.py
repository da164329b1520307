"""The Python calls of the state space scan and its convolution refuse wrong
arguments with KDAError (no GPU: nothing here reaches a launch)."""
import pytest

import gated_delta_rule_amd as kda

torch = pytest.importorskip("torch")

W, A = torch.zeros(64, 4), torch.zeros(2)
X, DT, B = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2), torch.zeros(1, 4, 1, 64)


@pytest.mark.parametrize("x", [None, 3.0, [1.0, 2.0], "x"])
@pytest.mark.parametrize("call", [lambda x: kda.ssm_conv_fwd(x, W), lambda x: kda.ssm_conv_step(x, W, None, None),
                                  lambda x: kda.ssm_conv_bwd(x, W, None, x), lambda x: kda.ssm_chunk_fwd(x, DT, A, B, B),
                                  lambda x: kda.ssm_chunk_bwd(x, DT, A, B, B, None, None, x),
                                  lambda x: kda.ssm_recurrent_fwd(x, DT, A, B, B, X)])
def test_x_is_no_tensor(call, x):
    with pytest.raises(kda.KDAError, match="x must be a torch.Tensor"):
        call(x)


def test_element_types_are_named():
    with pytest.raises(kda.KDAError, match="x must be bfloat16 or float32, got torch.float16"):
        kda.ssm_conv_fwd(torch.zeros(1, 4, 64).half(), W)
    with pytest.raises(kda.KDAError, match="x must be bfloat16 or float32, got torch.float64"):
        kda.ssm_chunk_fwd(X.double(), DT, A, B, B)


@pytest.mark.parametrize("other", ["dt", "A", "B", "C", "D", "S0", "cu_seqlens", "dt_bias"])
def test_other_arguments(other):
    ok = dict(x=X, dt=DT, A=A, B=B, C=B)
    with pytest.raises(kda.KDAError):
        kda.ssm_chunk_fwd(**{**ok, other: 3})
    for shape in ((), (4,), (4, 2)):
        with pytest.raises(kda.KDAError):
            kda.ssm_chunk_fwd(**{**ok, "x": torch.zeros(shape)})
