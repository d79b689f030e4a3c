"""Linear attention without any token: states pass through, gradients are empty or zero."""
import pytest
import torch

import gated_deltanet_fwd_amd as G

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("N", [1, 3])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_tokens(N, decay, dtype):
    H, HV, d = 1, 2, 64
    p = G.LinearProblem([0] * (N + 1), H, HV, d, dtype=dtype, decay=decay, has_h0=True, want_ht=True)
    q, v = torch.empty(0, H, d, dtype=dtype, device=DEV), torch.empty(0, HV, d, dtype=dtype, device=DEV)
    g = torch.zeros(HV, device=DEV) if decay == "head" else torch.empty(0, HV, device=DEV)
    cu = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    h0, dht = torch.randn(2, N, HV, d, d, device=DEV)
    o, ht = G.gdn_linear_fwd(p, q, q, v, g, cu, h0=h0)
    b = G.gdn_linear_bwd(p, q, q, v, g, cu, v, h0=h0, dht=dht)
    assert o.shape == v.shape and b["dq"].shape == q.shape and b["dv"].shape == v.shape and b["dg"].shape == g.shape
    assert torch.equal(ht, h0) and torch.equal(b["dh0"], dht) and not b["dg"].any()
