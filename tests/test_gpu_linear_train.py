"""A layer's gradients through the operators together: norm with the residual, projections, linear attention, the norm
of its output, in FP32, against 64-bit autograd of the formulas and against differences along random directions."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-6


def norm64(x, w):
    return w * x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()


class Layer:
    def __init__(self, lengths, C, H, HV, d, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
        self.cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        self.on_gpu, T = torch.from_numpy(self.cu).to(DEV), int(self.cu[-1])
        self.C, self.H, self.HV, self.d, self.scale = C, H, HV, d, d ** -0.5
        self.x = dict(x=normal(T, C), residual=normal(T, C), w=1 + 0.1 * normal(C), wo=1 + 0.1 * normal(HV * d),
                      proj=normal(C, (2 * H + HV) * d) / math.sqrt(C), gate=normal(C, HV) / math.sqrt(C))
        self.dy, self.dtotal = normal(T, HV * d), normal(T, C)  # gradients of the output and of the residual's stream

    def split(self, row):
        T, n = row.shape[0], self.H * self.d
        return row[:, :n].view(T, self.H, self.d), row[:, n:2 * n].view(T, self.H, self.d), row[:, 2 * n:].view(T, self.HV, self.d)

    def gradients(self):
        """Of the loss sum(dy out) + sum(dtotal total), by the framework's calls."""
        x, T = self.x, self.x["x"].shape[0]
        pn = G.RmsNormProblem(T, self.C, dtype=torch.float32, eps=EPS)
        po = G.RmsNormProblem(T, self.HV * self.d, dtype=torch.float32, eps=EPS)
        pl = G.LinearProblem(self.cu, self.H, self.HV, self.d, dtype=torch.float32, scale=self.scale)
        y, _, total = G.gdn_rms_norm_fwd(pn, x["x"], weight=x["w"], residual=x["residual"])
        row, z = y @ x["proj"], y @ x["gate"]
        q, k, v = self.split(row)
        g = torch.nn.functional.logsigmoid(z + 2)
        o, _ = G.gdn_linear_fwd(pl, q, k, v, g, self.on_gpu)
        o = o.view(T, -1)
        bo = G.gdn_rms_norm_bwd(po, o, self.dy, weight=x["wo"])
        b = G.gdn_linear_bwd(pl, q, k, v, g, self.on_gpu, bo["dx"].view(T, self.HV, self.d))
        drow = torch.cat([b[n].reshape(T, -1) for n in ("dq", "dk", "dv")], 1)
        dz = b["dg"] * torch.sigmoid(-z - 2)
        dy = drow @ x["proj"].T + dz @ x["gate"].T
        bn = G.gdn_rms_norm_bwd(pn, total, dy, weight=x["w"], d_residual=self.dtotal)
        return dict(x=bn["dx"], residual=bn["dx"], w=bn["dweight"], wo=bo["dweight"], proj=y.T @ drow, gate=y.T @ dz)

    def loss(self, x):
        """In 64 bits on the CPU, token by token pairs."""
        total = x["x"] + x["residual"]
        y = norm64(total, x["w"])
        q, k, v = self.split(y @ x["proj"])
        q, k = (t.repeat_interleave(self.HV // self.H, 1) for t in (q, k))
        g = torch.nn.functional.logsigmoid(y @ x["gate"] + 2)
        outs = []
        for b, e in zip(self.cu[:-1], self.cu[1:]):
            s = g[b:e].cumsum(0).T  # [HV, t]
            fade = (s[:, :, None] - s[:, None, :]).tril().exp().tril()
            p = torch.einsum("thd,shd->hts", q[b:e], k[b:e]) * fade
            outs.append(self.scale * torch.einsum("hts,shd->thd", p, v[b:e]).reshape(e - b, -1))
        out = norm64(torch.cat(outs), x["wo"])
        return (out * self.dy.double().cpu()).sum() + (total * self.dtotal.double().cpu()).sum()


# Sums of at most 2^9 terms, a rounding of 2^-24 each, through four products and two norms one after the other; a norm
# divides by the row's length, which keeps relative errors, but a row of o can be shorter than its terms by 2^4.
BOUND = 4 * 2.0 ** 4 * 2.0 ** 9 * 2.0 ** -24


@pytest.mark.parametrize("lengths,C,H,HV,d", [([70, 1, 129], 256, 2, 4, 64), ([300], 128, 1, 2, 128)])
def test_gradients_of_a_layer(lengths, C, H, HV, d):
    s = Layer(lengths, C, H, HV, d, 21)
    got = {n: t.double().cpu() for n, t in s.gradients().items()}
    leaves = {n: t.double().cpu().requires_grad_() for n, t in s.x.items()}
    s.loss(leaves).backward()
    for n, t in got.items():
        want = leaves[n].grad
        off = float((t - want).norm() / want.norm())
        print("%-8s off by %.2e" % (n, off))
        assert off <= BOUND, n
    # along a random direction: central differences of the 64-bit loss are off by h^2 times its third derivative
    gen = torch.Generator().manual_seed(2)
    with torch.no_grad():
        for n, t in got.items():
            u = torch.randn(t.shape, generator=gen, dtype=torch.float64)
            u *= leaves[n].norm() / u.norm()
            at = lambda h: float(s.loss({**leaves, n: leaves[n] + h * u}))  # noqa: E731
            h = 1e-5
            difference = (at(h) - at(-h)) / (2 * h)
            assert abs(difference - float((t * u).sum())) <= BOUND * float(t.norm() * u.norm()), n
