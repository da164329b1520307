"""The Python calls of softmax attention and its pages refuse wrong arguments
with KDAError (no GPU: nothing here reaches a launch)."""
import pytest

import gated_delta_rule_amd as kda

torch = pytest.importorskip("torch")

Q, K = torch.zeros(1, 4, 4, 64), torch.zeros(1, 4, 2, 64)
PAGES = torch.zeros(3, 2, 16, 64)
TABLE, LEN, REFS = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
LSE = torch.zeros(1, 4, 4)


@pytest.mark.parametrize("x", [None, 3.0, [1.0], "x", torch.zeros(4), torch.zeros(4, 64)])
@pytest.mark.parametrize("call", [lambda x: kda.attn_fwd(x, K, K), lambda x: kda.attn_fwd(Q, x, K), lambda x: kda.attn_fwd(Q, K, x),
                                  lambda x: kda.attn_bwd(x, K, K, Q, LSE, Q), lambda x: kda.attn_bwd(Q, K, K, x, LSE, Q),
                                  lambda x: kda.attn_paged_fwd(x, PAGES, PAGES, TABLE, LEN),
                                  lambda x: kda.attn_paged_fwd(Q, x, PAGES, TABLE, LEN),
                                  lambda x: kda.attn_paged_fwd(Q, PAGES, PAGES, x, LEN),
                                  lambda x: kda.kv_append(x, K, PAGES, PAGES, TABLE, LEN),
                                  lambda x: kda.kv_append(K, K, PAGES, PAGES, TABLE, x),
                                  lambda x: kda.kv_resize(x, LEN, REFS, LEN, 16), lambda x: kda.kv_resize(TABLE, LEN, REFS, x, 16),
                                  lambda x: kda.kv_fork(TABLE, LEN, REFS, x, LEN, PAGES, 16),
                                  lambda x: kda.kv_compact(TABLE, x, REFS, PAGES, 16)])
def test_wrong_arguments(call, x):
    with pytest.raises(kda.KDAError):
        call(x)


def test_host_tensors_and_types_are_refused():
    with pytest.raises(kda.KDAError, match="q must be a device tensor"):
        kda.attn_fwd(Q, K, K)
    with pytest.raises(kda.KDAError, match="q must be bfloat16 or float32, got torch.float16"):
        kda.attn_fwd(Q.half(), K, K)
    with pytest.raises(kda.KDAError, match="batch and token axes"):
        kda.attn_fwd(Q[0], K[0], K[0])
    with pytest.raises(kda.KDAError, match="k_pages must be a device tensor"):
        kda.attn_paged_fwd(Q, PAGES, PAGES, TABLE, LEN)
    with pytest.raises(kda.KDAError, match="table must be a device tensor"):
        kda.kv_resize(TABLE, LEN, REFS, LEN, 16)
