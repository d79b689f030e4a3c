"""Linear attention's segments in launches of more than 2^20 workgroups, which have two dimensions and so workgroups behind
the last one that has work: one document long enough for segments among tens of thousands of empty ones.

Bounds as in test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

DEV, K = "cuda:0", 600 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def close(name, got, ref, mag):
    x = got.double().cpu().numpy()
    bound = K * mag + (1.01 * 2.0 ** -8 * (np.abs(ref) + mag) if got.dtype == torch.bfloat16 else 0) + 1e-37
    assert x.shape == ref.shape and (np.abs(x - ref) <= bound).all(), name


@pytest.mark.parametrize("before,dtype", [(0, "bf16"), (30000, "f32"), (65534, "bf16")])
def test_workgroups_behind_the_last_segment(before, dtype):
    """The forward's states, one job in a launch of 1,048,624 workgroups and 2^20 - 48 more behind them."""
    H, d, T, N, scale = 16, 64, 1024, 65535, 0.11
    cu = np.zeros(N + 1, np.int32)
    cu[before + 1:] = T
    p = G.LinearProblem(cu, H, H, d, dtype=TYPES[dtype], scale=scale)
    # with segments, and in more than 2^20 workgroups that are no multiple of it: at most 256 tokens each
    slots = T // 256 + N
    assert slots * H > 1 << 20 and slots * H % (1 << 20)
    assert G.gdn_linear_workspace_bytes(p, 0) >= slots * H * (d * d + 1) * 4
    gen = torch.Generator(device=DEV).manual_seed(5)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    q, k, v = (normal(T, H, d).to(TYPES[dtype]) for _ in range(3))
    g = -torch.rand(T, H, generator=gen, device=DEV)
    print("forward of %d workgroups" % (slots * H), flush=True)
    o, _ = G.gdn_linear_fwd(p, q, k, v, g, torch.from_numpy(cu).to(DEV))
    x = [t.double().cpu().numpy() for t in (q, k, v, g)]
    A = [np.abs(t) for t in x[:3]]
    close("o", o, lo.fwd([0, T], *x, None, scale)[0], lo.fwd([0, T], *A, x[3], None, scale)[0])
