"""Linear attention, its step and the RMS norm at sizes where 32-bit offsets and one-dimensional launches end: what
lies behind them has the bits of (or, where the call is cut into other segments, is within the roundings of) a call
on that part alone."""
import numpy as np
import pytest
import torch

import gated_deltanet_fwd_amd as G

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def normal(gen, *s, dtype=torch.bfloat16):
    return torch.randn(*s, generator=gen, device=DEV, dtype=dtype)


def part(lengths, first):
    """Tokens and documents of the call on documents first .. alone."""
    t = sum(lengths[:first])
    cu = np.concatenate([[0], np.cumsum(lengths[first:])]).astype(np.int32)
    return t, cu


def run(lengths, H, HV, d, x, first=0):
    t, cu = part(lengths, first)
    on_gpu = torch.from_numpy(cu).to(DEV)
    p = G.LinearProblem(cu, H, HV, d, scale=0.1)
    a = [x[n][t:] for n in "qkvg"]
    o, _ = G.gdn_linear_fwd(p, *a, on_gpu)
    return dict(G.gdn_linear_bwd(p, *a, on_gpu, x["do"][t:]), o=o)


def inputs(T, H, HV, d):
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = dict(q=normal(gen, T, H, d), k=normal(gen, T, H, d), v=normal(gen, T, HV, d), do=normal(gen, T, HV, d))
    x["g"] = -torch.rand(T, HV, generator=gen, device=DEV)
    return x


def test_more_workgroups_than_one_dimension_holds():
    """65,535 documents and 96 heads: 18.9 million workgroups in the backward."""
    lengths = [1] * 65500 + [0, 3, 65] + [1] * 32
    x = inputs(sum(lengths), 32, 96, 64)
    whole, first = run(lengths, 32, 96, 64, x), 65400
    t, _ = part(lengths, first)
    last = run(lengths, 32, 96, 64, x, first)
    for name in ("o", "dq", "dk", "dv", "dg"):
        assert torch.equal(whole[name][t:], last[name]), name


def test_tokens_behind_32_bit_offsets():
    """2.2e9 values of v. Each side is within a rounding of P, of the state and of itself, 2^-8 at most each."""
    lengths = [269000, 1000]
    x = inputs(sum(lengths), 1, 64, 128)
    whole, last = run(lengths, 1, 64, 128, x), run(lengths, 1, 64, 128, x, 1)
    for name in ("o", "dq", "dk", "dv", "dg"):
        got, want = whole[name][269000:].double(), last[name].double()
        assert torch.isfinite(got).all()
        assert float((got - want).norm()) <= 6 * 2.0 ** -8 * float(want.norm()), name


def test_states_behind_32_bit_offsets():
    """A cache of 2.2e9 values; the step on its last slots is the step on a cache of those alone."""
    n, H, HV, d, N = 2800, 16, 48, 128, 5
    gen = torch.Generator(device=DEV).manual_seed(4)
    states = torch.zeros(n, HV, d, d, device=DEV)
    few = normal(gen, 2 * N, HV, d, d, dtype=torch.float32)
    states[-2 * N:] = few
    lengths = [2, 1, 0, 3, 1]
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T, on_gpu = int(cu[-1]), torch.from_numpy(cu).to(DEV)
    q, k, v = normal(gen, T, H, d), normal(gen, T, H, d), normal(gen, T, HV, d)
    g = -torch.rand(T, HV, generator=gen, device=DEV)
    slot = torch.arange(N, dtype=torch.int32, device=DEV)
    keep = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    keep[0] = 2 * N - 1
    outs = []
    for cache, base in ((states, n - 2 * N), (few, 0)):
        p = G.LinearStepProblem(N, H, HV, d, cache.shape[0], cu_seqlens_host=cu)
        at = torch.where(keep < 0, keep, keep + base)
        outs.append(G.gdn_linear_step(p, q, k, v, g, cache, slot + base, slot + base + N - 1, slot_tok=at, cu_seqlens=on_gpu))
    assert torch.equal(*outs) and torch.equal(states[-2 * N:], few)
    assert not states[:-2 * N].any()


@pytest.mark.parametrize("rows,d,out", [(70_000_001, 8, "io"), (135_001, 16384, "e4m3")])
def test_norm_rows(rows, d, out):
    """More workgroups of 256 threads than one dimension holds; 2.2e9 values."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, few = normal(gen, rows, d), 1001
    w = 1 + 0.1 * normal(gen, d, dtype=torch.float32)
    plan = lambda n: G.RmsNormProblem(n, d, out=out)  # noqa: E731
    whole = G.gdn_rms_norm_fwd(plan(rows), x, weight=w, residual=x)
    last = G.gdn_rms_norm_fwd(plan(few), x[-few:].clone(), weight=w, residual=x[-few:].clone())
    for a, b in zip(whole, last):
        if a is not None:
            assert torch.equal(a[-few:].view(torch.uint8), b.view(torch.uint8))
    if out == "io":
        y = x[:few].double() * 2
        y = w.double() * y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        assert ((whole[0][:few].double() - y).abs() <= 1.01 * 2.0 ** -8 * y.abs()).all()
        grads = [G.gdn_rms_norm_bwd(plan(n), x[-n:], x[-n:], weight=w)["dx"] for n in (rows, few)]
        assert torch.equal(grads[0][-few:], grads[1])
