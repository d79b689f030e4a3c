"""RMS norm with the residual's addition on MI355X against float64, forward (io and 8 bits) and backward.

Bounds: r = 1 / sqrt(mean x^2 + eps) sums up to 16,384 squares (a lane adds at most 64, the lanes' sums meet in at most 10
steps) and rounds a few times more: under 60 roundings of 2^-24, so f32 results are held to 60 2^-24 of their value
(the sum x + r: one rounding; gradients: of the magnitudes that are added). bf16 results add 2^-8 of their value. 8-bit values are
held to half a step at the scaled value, 2^-4 of it or 2^-10 below 2^-6, beside the f32 bound; scales to the f32 bound.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G

pytestmark = pytest.mark.gpu

DEV, K = "cuda:0", 60 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def close(name, got, ref, mag=None):
    mag = ref.abs() if mag is None else mag
    bound = K * mag + (2.0 ** -8 * ref.abs() if got.dtype == torch.bfloat16 else 0) + 1e-37
    off = (got.double() - ref).abs() - bound
    assert got.shape == ref.shape and bool((off <= 0).all()), (name, float(off.max()))


def inputs(rows, d, dtype, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    wide = torch.randn(rows, 2 * d + 8, generator=gen, device=DEV).to(TYPES[dtype])
    return wide[:, :d], wide[:, d:2 * d], 1 + 0.1 * torch.randn(d, generator=gen, device=DEV), gen


SIZES = [(1, 8), (3, 64), (5, 520), (2, 1000), (7, 2048), (1500, 2048), (1025, 1016), (3, 4096), (2, 8192), (3, 10240), (2, 16384)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False)])
def test_forward_and_backward(rows, d, dtype, residual, weight):
    x, r, w, gen = inputs(rows, d, dtype)
    r, w = r if residual else None, w if weight else None
    p = G.RmsNormProblem(rows, d, dtype=TYPES[dtype], eps=1e-5)
    y, scales, out = G.gdn_rms_norm_fwd(p, x, weight=w, residual=r)
    t = x.double() + r.double() if residual else x.double()
    W = w.double() if weight else torch.ones(d, dtype=torch.float64, device=DEV)
    inv = 1 / ((t ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
    mag = x.double().abs() + r.double().abs() if residual else t.abs()
    close("y", y, t * inv * W, mag * inv * W.abs())
    assert scales is None and (out is None) == (not residual)
    if residual:
        close("residual_out", out, t, mag)
    dy = torch.randn(rows, d, generator=gen, device=DEV).to(TYPES[dtype])
    b = G.gdn_rms_norm_bwd(p, x, dy, weight=w, d_residual=r)
    t = x.double()
    inv = 1 / ((t ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
    n, dn = t * inv, dy.double() * W
    m, mA = (n * dn).mean(-1, keepdim=True), (n * dn).abs().mean(-1, keepdim=True)
    plus = r.double() if residual else torch.zeros_like(t)
    close("dx", b["dx"], inv * (dn - n * m) + plus, 3 * (inv * (dn.abs() + n.abs() * mA) + plus.abs()))
    if weight:  # rows are summed one after the other in a workgroup
        part = dy.double() * n
        bound = (60 + rows / 512 + 40) * 2.0 ** -24 * part.abs().sum(0)
        assert bool(((b["dweight"].double() - part.sum(0)).abs() <= bound + 1e-37).all())
    else:
        assert b["dweight"] is None


@pytest.mark.parametrize("rows,d", [(1, 128), (3, 640), (1100, 2048), (2, 4096), (5, 10240), (2, 16384)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_eight_bits(rows, d, group, dtype):
    x, r, w, _ = inputs(rows, d, dtype, seed=2)
    x[0] = 0
    if rows > 1:
        r = r.clone()
        x[1, :32] = 0
        r[1, :32] = 0  # a group of zeros (whole only where group = 32)
        r[0] = 0       # and a row
    p = G.RmsNormProblem(rows, d, dtype=TYPES[dtype], out="e4m3", group=group)
    res = r if rows > 1 else None
    y, scales, out = G.gdn_rms_norm_fwd(p, x, weight=w, residual=res)
    t = x.double() + (res.double() if res is not None else 0)
    ref = t / ((t ** 2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    mag = (x.double().abs() + (res.double().abs() if res is not None else 0)) / ((t ** 2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double().abs()
    z, zm = (v.view(rows, -1, group or d) for v in (ref, mag))
    most = z.abs().amax(-1)
    assert y.dtype == torch.float8_e4m3fn and scales.shape == most.shape
    zero = most == 0
    assert bool((scales[zero] == 1).all()) and bool(zero[0].all())
    # the largest magnitude may be of a sum that cancels: the bound of what was added
    off = (scales.double() * 448 - most).abs() - K * 2 * zm.amax(-1)
    assert bool((off[~zero] <= 0).all())
    s = scales.double()[..., None]
    got, want = y.double().view_as(z), z / s
    bound = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) + 2 * K * (zm / s + want.abs())
    assert bool(((got - want).abs() <= bound).all())
    assert float(y.double().abs().max()) <= 448


def test_eight_bits_are_the_nearest():
    """Values whose scaled forms are exact: every e4m3 value and the midpoints, ties to even."""
    e4m3 = torch.arange(0, 0x7f, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).float()
    mids = (e4m3[1:] + e4m3[:-1]) / 2
    row = torch.cat([e4m3, mids, -e4m3[1:4]])[:256]
    row = torch.cat([row, row.new_zeros(256 - row.numel())])
    row[-1] = 448.0
    # weights carry the values; a row of ones has the norm 1 with eps = 0
    p = G.RmsNormProblem(1, 256, dtype=torch.float32, out="e4m3", eps=0.0)
    y, scales, _ = G.gdn_rms_norm_fwd(p, torch.ones(1, 256, device=DEV), weight=row)
    assert float(scales) == 1.0
    assert torch.equal(y.float()[0], row.clamp(-448, 448).to(torch.float8_e4m3fn).float())


def test_rows_that_are_not_finite_stay_alone():
    for out in ("io", "e4m3"):
        x, r, w, _ = inputs(6, 512, "f32", seed=3)
        p = G.RmsNormProblem(6, 512, dtype=torch.float32, out=out)
        want = G.gdn_rms_norm_fwd(p, x, weight=w, residual=r)
        x = x.clone()
        x[2, 7], x[4, 500] = float("nan"), float("inf")
        got = G.gdn_rms_norm_fwd(p, x, weight=w, residual=r)
        rest = [0, 1, 3, 5]
        for a, b in zip(want, got):
            if a is not None:
                assert torch.equal(a.float()[rest], b.float()[rest])
        assert torch.isnan(got[0].float()[2]).all() and torch.isnan(got[0].float()[4, 500])


def test_subnormal_rows_and_zeros():
    """Mean squares below FP32's normal numbers, eps = 0: the row is still normalised; zeros with eps give zeros."""
    p = G.RmsNormProblem(2, 64, dtype=torch.float32, eps=0.0)
    x = torch.randn(2, 64, device=DEV)
    x[1] *= 2.0 ** -66
    y = G.gdn_rms_norm_fwd(p, x)[0]
    ref = x.double() / (x.double() ** 2).mean(-1, keepdim=True).sqrt()
    assert float((y[0].double() - ref[0]).abs().max()) < 1e-5
    assert float((y[1].double() - ref[1]).abs().max()) < 2.0 ** -6  # squares of 2^-132 keep few bits (149 - 132 less 6 for the mean)
    z = G.gdn_rms_norm_fwd(G.RmsNormProblem(2, 64, dtype=torch.float32), torch.zeros(2, 64, device=DEV))[0]
    assert bool((z == 0).all())


def test_no_rows_given_buffers_and_in_place():
    p = G.RmsNormProblem(0, 64)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    assert G.gdn_rms_norm_fwd(p, e, weight=w, residual=e)[0].shape == (0, 64)
    b = G.gdn_rms_norm_bwd(p, e, e, weight=w)
    assert b["dx"].shape == (0, 64) and bool((b["dweight"] == 0).all())
    x, r, w, _ = (t.contiguous() if torch.is_tensor(t) else t for t in inputs(9, 1024, "bf16"))
    p = G.RmsNormProblem(9, 1024)
    y, _, out = G.gdn_rms_norm_fwd(p, x, weight=w, residual=r)
    x2, r2 = x.clone(), r.clone()
    y2, _, out2 = G.gdn_rms_norm_fwd(p, x2, weight=w, residual=r2, y=x2, residual_out=r2)
    assert y2 is x2 or y2.data_ptr() == x2.data_ptr()
    assert torch.equal(y, x2) and torch.equal(out, r2)
    g = G.gdn_rms_norm_bwd(p, x, y, weight=w, d_residual=r)
    y3 = y.clone()
    g2 = G.gdn_rms_norm_bwd(p, x, y3, weight=w, d_residual=r, grads=dict(dx=y3))
    assert torch.equal(g["dx"], y3) and torch.equal(g["dweight"], g2["dweight"])


def test_graph_and_stream():
    x, r, w, gen = inputs(300, 2048, "bf16", seed=5)
    p, q = G.RmsNormProblem(300, 2048, out="e4m3", group=128), G.RmsNormProblem(300, 2048)
    dy = torch.randn(300, 2048, generator=gen, device=DEV).bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s, out = G.gdn_rms_norm_fwd(p, x, weight=w, residual=r)
        b = G.gdn_rms_norm_bwd(q, out, dy, weight=w, d_residual=r)
    side = torch.cuda.Stream()
    for _ in range(3):
        x.mul_(-0.7)
        dy.add_(0.1)
        side.wait_stream(torch.cuda.current_stream())
        y2, s2, out2 = G.gdn_rms_norm_fwd(p, x, weight=w, residual=r, stream=side)
        b2 = G.gdn_rms_norm_bwd(q, out2, dy, weight=w, d_residual=r, stream=side)
        side.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.float(), y2.float()) and torch.equal(s, s2) and torch.equal(out, out2)
        assert torch.equal(b["dx"], b2["dx"]) and torch.equal(b["dweight"], b2["dweight"])


def test_binding_refusals():
    x, r, w, _ = inputs(4, 64, "bf16")
    p = G.RmsNormProblem(4, 64)
    for a, kw in (((x[:3],), {}), ((x.float(),), {}), ((x,), dict(weight=w.bfloat16())), ((x,), dict(residual=r[:, :32])),
                  ((x,), dict(scales=torch.zeros(4, 1, device=DEV))), ((x,), dict(residual_out=r)), ((x.t(),), {})):
        with pytest.raises(G.GdnError):
            G.gdn_rms_norm_fwd(p, *a, **kw)
    with pytest.raises(G.GdnError):
        G.gdn_rms_norm_bwd(p, x, x[:2])
    with pytest.raises(G.GdnError):
        G.gdn_rms_norm_bwd(G.RmsNormProblem(4, 64, out="e4m3"), x, x.contiguous())
