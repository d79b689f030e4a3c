"""Rising decays: log decays whose sums over a chunk stay in FP32's range and over a segment do not, on states that are zero
there: what the segments' states are joined with must leave zeros zeros.

Bounds as in test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
import linear_util as u
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

DEV, K = "cuda:0", 600 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
T, D, LIVE, SCALE = 4096, 64, 50, 0.2


def close(name, got, ref, mag):
    x = got.double().cpu().numpy()
    bound = K * mag + (1.01 * 2.0 ** -8 * (np.abs(ref) + mag) if got.dtype == torch.bfloat16 else 0) + 1e-37
    assert (np.abs(x - ref) <= bound).all(), name  # (a NaN is not)


def inputs(dtype):
    q, k, v, _, do, _, _ = u.dg_inputs([T], 1, 1, D, "token", False, False, 9)
    g = np.random.default_rng(2).uniform(0.8, 1.2, (T, 1)).astype(np.float32)
    # in range over every 64 tokens, past it over every 128
    sums = np.concatenate([[0], np.cumsum(g.astype(np.float64))])
    assert (sums[64:] - sums[:-64]).max() < 80 and (sums[128:] - sums[:-128]).min() > 95
    p = G.LinearProblem([0, T], 1, 1, D, dtype=TYPES[dtype], scale=SCALE, want_ht=True)
    on = lambda x: torch.from_numpy(x).to(DEV).to(TYPES[dtype])  # noqa: E731
    return q, k, v, do, g, p, on, torch.from_numpy(g).to(DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(dtype):
    """Keys of zeros but for the last tokens'."""
    q, k, v, _, g, p, on, gg, cu = inputs(dtype)
    k[:T - LIVE] = 0
    slots = T // 128 + 1  # segments of at most 128 tokens would not overflow: the plan has those of 128
    assert G.gdn_linear_workspace_bytes(p, G.OP_FWD) == (slots * D * D * 4 + 255) // 256 * 256 + (slots * 4 + 255) // 256 * 256
    o, ht = G.gdn_linear_fwd(p, on(q), on(k), on(v), gg, cu)
    a = [x.astype(np.float64) for x in (q, k, v)]
    ref, kept = lo.steps([0, T], *a, g.astype(np.float64), None, SCALE)
    A, keptA = lo.steps([0, T], *[np.abs(x) for x in a], g.astype(np.float64), None, SCALE)
    close("o", o, ref, A)
    close("ht", ht[0], kept[-1], keptA[-1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(dtype):
    """Output gradients of zeros but for the first tokens', keys of zeros (the states themselves would leave FP32's range)."""
    q, k, v, do, g, p, on, gg, cu = inputs(dtype)
    k[:] = 0
    do[LIVE:] = 0
    assert u.backward_is_cut(p, 1, 1, D, dtype)
    b = G.gdn_linear_bwd(p, on(q), on(k), on(v), gg, cu, on(do))
    dk, dkA, S, SA = np.zeros((T, 1, D)), np.zeros((T, 1, D)), np.zeros((D, D)), np.zeros((D, D))
    for t in range(LIVE - 1, -1, -1):
        x = SCALE * np.outer(q[t, 0].astype(np.float64), do[t, 0].astype(np.float64))
        S, SA = S + x, SA + np.abs(x)
        dk[t, 0], dkA[t, 0] = S @ v[t, 0], SA @ np.abs(v[t, 0])
        S, SA = S * np.exp(np.float64(g[t, 0])), SA * np.exp(np.float64(g[t, 0]))
    close("dk", b["dk"], dk, dkA)
    for x in ("dq", "dv", "dg"):
        assert not b[x].any(), x
