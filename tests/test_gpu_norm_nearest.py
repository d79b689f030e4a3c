"""The norm's 8-bit output is the value nearest to x / scale, ties to even, also beside the midpoints of two 8-bit values and
with scales that are no powers of two. Which one is nearest is decided without rounding: an FP32 value and a scale times a
midpoint (24 + 5 bits) are float64 numbers, and so is their difference here."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GRID = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()  # 0 .. 448, rising
MIDS = (GRID[1:] + GRID[:-1]) / 2


def nearest(v, s):
    """Of GRID and its negatives, by exact comparisons with scaled midpoints; ties to the even code."""
    m = np.abs(v)
    code = (m[:, None] > s[:, None] * MIDS).sum(1)
    tie = (m[:, None] == s[:, None] * MIDS).any(1)
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    return np.sign(v) * GRID[code]


def values(d, group, r):
    """Groups of values beside midpoints, up to two FP32 steps off, at scales from 2^-60 to 2^60."""
    w = np.zeros(d, np.float32)
    for at in range(0, d, group):
        most = np.float32(r.uniform(1, 2) * 2.0 ** r.integers(-60, 60))
        s = np.float32(most) / np.float32(448)
        near = (r.choice(MIDS, group) * np.float64(s)).astype(np.float32)
        near = (near.view(np.int32) + r.integers(-2, 3, group).astype(np.int32)).view(np.float32)
        w[at:at + group] = near * r.choice([-1, 1], group)
        w[at + r.integers(group)] = most
    return w


@pytest.mark.parametrize("d,group", [(256, 0), (8192, 32), (2048, 64), (16384, 128), (4096, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nearest_beside_midpoints(d, group, dtype):
    w = values(d, group or d, np.random.default_rng(d + group))
    # weights carry the values: a row of ones has the norm 1 with eps = 0
    p = G.RmsNormProblem(3, d, dtype=dtype, out="e4m3", group=group, eps=0.0)
    y, scales, _ = G.gdn_rms_norm_fwd(p, torch.ones(3, d, dtype=dtype, device=DEV), weight=torch.from_numpy(w).to(DEV))
    most = np.abs(w).reshape(-1, group or d).max(1)
    assert torch.equal(scales.cpu(), torch.from_numpy(most / np.float32(448)).expand(3, -1))
    want = nearest(w.astype(np.float64), np.repeat((most / np.float32(448)).astype(np.float64), group or d))
    for row in y.double().cpu().numpy():
        assert (row == want).all(), int((row != want).sum())
    # one rounding too many would show: the rounded quotient's nearest is another one here and there
    q = torch.from_numpy((w.reshape(len(most), -1) / (most / np.float32(448))[:, None]).ravel())
    assert (q.to(torch.float8_e4m3fn).double().numpy() != want).any()


def test_infinite_and_absent_scales():
    """An infinite value makes its group's scale infinite: finite values over it are 0, with their signs, and it is NaN
    itself; other groups stay. A group of zeros is zeros with the scale 1."""
    w = torch.ones(96, device=DEV)
    w[3], w[4], w[5] = float("inf"), -2.0, 0.0
    w[32:64] = 0
    p = G.RmsNormProblem(1, 96, dtype=torch.float32, out="e4m3", group=32, eps=0.0)
    y, scales, _ = G.gdn_rms_norm_fwd(p, torch.ones(1, 96, device=DEV), weight=w)
    assert scales.tolist()[0][:2] == [float("inf"), 1.0]
    y = y.float()[0]
    assert torch.isnan(y[3]) and bool((y[:3] == 0).all()) and bool((y[4:64] == 0).all()) and bool((y[64:] == 448).all())
