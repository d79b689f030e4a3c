"""Decays whose factor is 0: the document is two, in every gradient, and the decay's own gradient is exactly 0."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
import linear_util as u
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("T,at", [(200, 90), (200, 0), (200, 199), (1500, 700), (1500, 1024)])
@pytest.mark.parametrize("value", [float("-inf"), -20000.0, -200.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("states", [True, False])
def test_gradient_of_a_dropped_state(T, at, value, dtype, states):
    H, HV, d, scale, dt = 1, 2, 64, 0.11, TYPES[dtype]
    q, k, v, g, do, h0, dht = u.dg_inputs([T], H, HV, d, "token", states, states, T + at)
    g[at] = value
    on = lambda x, t=torch.float32: None if x is None else torch.from_numpy(x).to(DEV).to(t)  # noqa: E731
    p = G.LinearProblem([0, T], H, HV, d, dtype=dt, scale=scale, has_h0=states)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    b = G.gdn_linear_bwd(p, on(q, dt), on(k, dt), on(v, dt), on(g), cu, on(do, dt), h0=on(h0), dht=on(dht))
    dg = b["dg"].double().cpu().numpy()
    assert (dg[at] == 0).all()
    # in 64 bits: two documents, of which the second begins without a state and the first leaves none
    g64 = g.astype(np.float64)
    g64[at] = -1.0
    N = np.zeros((1, HV, d, d))
    two = lambda x, first: None if x is None else np.concatenate([x, N] if first else [N, x])  # noqa: E731
    a = [x.astype(np.float64) for x in (q, k, v)]
    ref, rows, norms = lo.dg_by_states([0, at, T], *a, g64, do.astype(np.float64), two(h0, True), two(dht, False), scale)
    # roundings of the row products on both sides of the drop meet in the sums of its segment
    bound = u.dg_bounds([0, T], rows, norms, d, False, u.most_tokens(dtype, "token"))[0]
    for part in (slice(0, at), slice(at + 1, T)):
        if part.start < part.stop:
            off = float(np.sqrt(((dg[part] - ref[part]) ** 2).mean()))
            assert off <= bound * np.sqrt(T / (part.stop - part.start)), (part, off, bound)


def test_one_decay_a_head_drops_all():
    """g = -inf for a head: its gradient is exactly 0, other heads' is what it is without it."""
    H, HV, d, T = 1, 3, 64, 700
    q, k, v, g, do, _, _ = u.dg_inputs([T], H, HV, d, "head", False, False, 5)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    p = G.LinearProblem([0, T], H, HV, d, dtype=torch.float32, decay="head")
    a = [torch.from_numpy(x).to(DEV) for x in (q, k, v)]
    outs = []
    for first in (float(g[0]), float("-inf")):
        g[0] = first
        outs.append(G.gdn_linear_bwd(p, *a, torch.from_numpy(g).to(DEV), cu, torch.from_numpy(do).to(DEV)))
    assert float(outs[1]["dg"][0]) == 0.0 and torch.equal(outs[0]["dg"][1:], outs[1]["dg"][1:])
    assert float(outs[0]["dg"][0]) != 0.0
